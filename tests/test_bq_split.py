"""CPU model of how the block-scaled decode cuts its work: every iteration of every
(sequence, kv head) is done once, every cut piece is joined from all its parts and
only those, and nothing lies outside the workspace."""
import random
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "paged_kv_cache_251_gb300" / "csrc"


def constant(name):
    for f in ("pa_decode_bq.cuh", "pa_block_quant.h"):
        m = re.search(rf"constexpr int {name} = (\d+);", (CSRC / f).read_text())
        if m:
            return int(m.group(1))
    raise AssertionError(name)


COST, SHARE = constant("kPieceCost"), constant("kMinShare")
THREADS = constant("kDecodeBqThreads")
WARPS = THREADS // 32
MAX_CTAS = constant("kDecodeBqSms") * constant("kDecodeBqCtas")


def ctas_of(seqs, hkv, max_len):
    iters = (max_len + 15) // 16 + COST
    per_cta = WARPS * (SHARE + COST)
    if seqs * hkv > MAX_CTAS * per_cta // iters:
        return MAX_CTAS
    return (seqs * hkv * iters + per_cta - 1) // per_cta


def run(tiles, hkv, u, ctas):
    """The kernel's arithmetic; returns what was done of each piece and how it is joined."""
    units = [(n + u - 1) // u + COST for n in tiles]
    total = hkv * sum(units)
    nwarps = ctas * WARPS
    share = max((total + nwarps - 1) // nwarps, SHARE + COST)
    assert share * nwarps >= total
    per = (len(tiles) + THREADS - 1) // THREADS
    prefix = [0]
    for t in range(THREADS):
        prefix.append(prefix[-1] + sum(hkv * units[s] for s in range(t * per, min((t + 1) * per, len(tiles)))))
    done, zeros, records, final, slots, last = {}, set(), {}, {}, {}, {}
    for wid in range(nwarps):
        u0, u1 = wid * share, min(wid * share + share, total)
        if u0 >= total:
            continue
        a, b = 0, THREADS
        while b - a > 1:
            m = (a + b) >> 1
            a, b = (m, b) if prefix[m] <= u0 else (a, m)
        seq, at = a * per, prefix[a]
        while at + hkv * units[seq] <= u0:
            at += hkv * units[seq]
            seq += 1
        head = (u0 - at) // units[seq]
        piece = at + head * units[seq]
        while True:
            iters = units[seq] - COST
            i0, i1 = u0 - piece - COST, u1 - piece - COST
            k0 = min(i0, iters) if i0 > 0 else 0
            k1 = max(i1, 0) if i1 < iters else iters
            if iters == 0 and u0 <= piece:
                assert (seq, head) not in zeros
                zeros.add((seq, head))
            if k0 < k1:
                done.setdefault((seq, head), []).append((k0, k1))
                if k0 == 0 and k1 == iters:
                    assert (seq, head) not in final
                    final[seq, head] = [(0, iters)]
                else:
                    assert (wid, int(k0 == 0)) not in slots
                    slots[wid, int(k0 == 0)] = (seq, head, k0, k1, k1 == iters)
                    if k0 == 0:
                        last[wid] = (piece + units[seq] - 1) // share // WARPS
            piece += units[seq]
            if piece >= u1:
                break
            head += 1
            if head == hkv:
                head, seq = 0, seq + 1
    parts = {}
    for cta in range(ctas):
        for w in range(WARPS):
            for first in ((0, 1) if w == 0 else (1,)):
                slot = slots.get((cta * WARPS + w, first))
                if slot is None:
                    continue
                got, ends, n = [slot], first == 0 and slot[4], 1
                while not ends and w + n < WARPS:
                    nxt = slots[cta * WARPS + w + n, 0]
                    assert nxt[:2] == slot[:2]
                    got.append(nxt)
                    ends = nxt[4]
                    n += 1
                ranges = [x[2:4] for x in got]
                if first == 1 and ends:
                    assert slot[:2] not in final
                    final[slot[:2]] = ranges
                else:
                    assert (cta, first) not in parts
                    parts[cta, first] = (slot[:2], ranges)
                    if first == 1:
                        assert cta not in records
                        records[cta] = (slot[:2], last[cta * WARPS + w])
    for cta, (pair, end) in records.items():
        assert cta < end < ctas and pair not in final
        got = []
        for c in range(cta, end + 1):
            who, ranges = parts.pop((c, int(c == cta)))
            assert who == pair
            got += ranges
        final[pair] = got
    assert not parts
    return done, zeros, final


@pytest.mark.parametrize("u", [1, 2])
def test_every_iteration_once(u):
    rng = random.Random(7)
    for case in range(120):
        seqs = rng.choice([1, 2, 3, 17, 255, 256, 257, 600])
        hkv = rng.choice([1, 2, 8])
        top = rng.choice([0, 1, 5, 60, 700 if seqs < 20 else 30])
        tiles = [rng.choice([0, rng.randint(0, top), top]) for _ in range(seqs)]
        most = ctas_of(seqs, hkv, 16 * max(max(tiles), 1))
        for ctas in {most, min(most, rng.randint(1, MAX_CTAS)), min(most, 152)}:
            done, zeros, final = run(tiles, hkv, u, ctas)
            for s, n in enumerate(tiles):
                iters = (n + u - 1) // u
                for h in range(hkv):
                    if iters == 0:
                        assert (s, h) in zeros and (s, h) not in done and (s, h) not in final
                        continue
                    for ranges in (done[s, h], final[s, h]):
                        ranges = sorted(ranges)
                        assert ranges[0][0] == 0 and ranges[-1][1] == iters
                        assert all(a[1] == b[0] for a, b in zip(ranges, ranges[1:]))


def test_one_cta_needs_no_join():
    """The join kernel is left out when there is one CTA: it holds every piece whole."""
    for seqs, hkv, tiles in ((1, 1, 80), (8, 1, 8), (2, 2, 19), (29, 1, 0)):
        if ctas_of(seqs, hkv, 16 * max(tiles, 1)) == 1:
            run([tiles] * seqs, hkv, 1, 1)
