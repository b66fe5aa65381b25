"""What the attention kernels' sources have to hold where no run shows it: a
missing order between two CTAs' accesses, or a warp that is not converged, goes
well until it does not.  Read from the sources, without a GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_attention_prolog_gb300", "csrc")


def code(name, start=None, end=None):
    """A source, or what lies between two of its role headings, without comments."""
    src = open(os.path.join(CSRC, name)).read()
    if start:
        a = src.index(start)
        src = src[a:src.index(end, a)]
    return " ".join(re.sub(r"//[^\n]*", "", src).split())


@pytest.mark.parametrize("name", ["attend_cache8_pair.cu", "attend_cache.cu"])
def test_copies_come_before_the_other_ctas_clears(name):
    """Rows behind a sequence's end are cleared by each CTA of a pair over rows that
    a copy brought, which the even CTA's barrier counted: its arrival at the odd one
    releases, and both looks acquire, at the scope of the cluster."""
    seen = code("attend_ptx.cuh")
    a = seen.index("void copies_seen(uint32_t full, uint32_t parity, uint32_t seen) {")
    assert [x for _, x in statements(seen[seen.index("{", a):seen.index("}", a)])] == [
        "mbar_acquire_cluster(full, parity)", "mbar_arrive(seen)", "mbar_arrive_cluster(map_shared_rank(seen, 1))"]
    src = code(name)
    at = [m.start() for m in re.finditer(r"smem_u32\(&sh->v_seen\)\);", src) if not src[:m.start()].endswith("acquire_cluster(")]
    assert at
    for a in at:
        told = src.rindex("copies_seen(smem_u32(&sh->v_full[", 0, a)
        assert ";" not in src[told:a] and told > src.rindex("look(&sh->v_full[", 0, a)
    waits = [m.end() for m in re.finditer(r"wait\(&sh->v_seen, tails\)", src)]
    assert waits
    for a in waits:
        behind = src[a:]
        assert behind.index("mbar_acquire_cluster(smem_u32(&sh->v_seen), tails & 1)") < behind.index("st_shared_v4(")


def statements(src):
    """(depth of braces, statement) in the order of the source; a block's head is a statement of the depth around it."""
    out, depth, inner, now = [], 0, 0, ""
    for c in src:
        inner += {"(": 1, ")": -1}.get(c, 0)
        if c in "{}" or (c == ";" and inner == 0):
            if now.strip():
                out.append((depth, now.strip()))
            now = ""
            depth += {"{": 1, "}": -1}.get(c, 0)
        else:
            now += c
    return out


COLLECTIVE = re.compile(r"\b(tmem_ld\w*|tmem_st\w*|get_o)\(")
CONVERGES = re.compile(r"__syncwarp\(|named_bar_(sync|or)\(|__\w+_sync\(|sum_across\(|arrive_even\(|" + COLLECTIVE.pattern)
DIVIDES = re.compile(r"\b(if|for) \(.*\b(lane|tid|threadIdx|mine|rows|r|column)\b")
LOOP = re.compile(r"\b(for|while) ?\(")


@pytest.mark.parametrize("name,start,end,least", [
    ("attend_cache8.cu", "- softmax\n", "- MMA\n", 7), ("attend_cache8_pair.cu", "- softmax\n", " MMA (the even CTA's", 5)])
def test_warps_are_converged_at_every_access_to_tensor_memory(name, start, end, least):
    """tcgen05.ld and .st take a whole converged warp: between one of them and what some lanes alone do (in front of it,
    or at the end of the round of the loop before) lies something that the whole warp has to come to."""
    code_ = statements(code(name, start, end))
    found = 0
    for i, (depth, s) in enumerate(code_):
        if not COLLECTIVE.search(s) or s.startswith("auto get_o") or "float (&o)[8]) " in s:
            continue
        found += 1
        # the innermost loop around it
        head, d = i - 1, depth
        while head >= 0 and not (code_[head][0] < d and LOOP.search(code_[head][1])):
            d = min(d, code_[head][0])
            head -= 1
        last = i
        while last + 1 < len(code_) and head >= 0 and code_[last + 1][0] > code_[head][0]:
            last += 1
        for s2 in [x for _, x in code_[head + 1:i][::-1]] + [x for _, x in code_[i + 1:last + 1][::-1]]:
            if CONVERGES.search(s2):
                break
            assert not DIVIDES.search(s2), f"`{s}` behind `{s2}`"
    assert found >= least


LEAVES = re.compile(r"^if \(!ok\) (continue|break)|^if \(failed\)|^if \(!?named_bar_or\(1, kSoft, .*!ok\)\)|^if \(ok( &&|\)) |"
                    r"r < kHeads && ok|\) scratch->failed\[warp\] = !ok")
EFFECT = re.compile(r"\b(tmem_st\w*|st_shared_v\d|mbar_arrive\w*|arrive_even)\(|\bsh->(m|by)\[.*\] [-*]?= |\bscratch->sum\[")


@pytest.mark.parametrize("name,start,end,least", [
    ("attend_cache8.cu", "- softmax\n", "- MMA\n", 6), ("attend_cache8_pair.cu", "- softmax\n", " MMA (the even CTA's", 6)])
def test_a_failed_wait_of_the_softmax_warps_stays_failed(name, start, end, least):
    """A wait that gave up is not forgotten when a later one succeeds, and what depends on it (a bound moved, O scaled, P
    overwritten, rows cleared, arrivals that hand them over) is not done: the warp leaves, or tells the others, before."""
    code_ = [s for _, s in statements(code(name, start, end))]
    waits = [i for i, s in enumerate(code_) if re.search(r"\bok = ", s) and "wait(" in s]
    assert len(waits) >= least
    for i in waits:
        assert re.search(r"\bok && wait\(", code_[i]), f"`{code_[i]}` forgets an earlier wait"
        leaves = next(j for j in range(i + 1, len(code_)) if LEAVES.search(code_[j]))
        done = [s for s in code_[i + 1:leaves] if EFFECT.search(s)]
        assert not done, f"after `{code_[i]}`: {done}"
    # the shared word that tells them is looked at behind a barrier, before what it guards
    told = next(i for i, s in enumerate(code_) if "scratch->failed[warp] = !ok" in s)
    known = next(i for i, s in enumerate(code_) if s.startswith("if (failed) break"))
    assert any("named_bar_sync(1, kSoft)" in s for s in code_[told:known])
    assert not [s for s in code_[told:known] if re.search(r"\b(tmem_st\w*|mbar_arrive\w*|arrive_even)\(", s)]


def ring(slots, chunks, blocks, early, steps=60):
    """The ring of attend_cache8.cu: two warps copy chunks of key steps into its places, a step's first two and the others, and
    wait for a place by the parity of its phase.  The tensor core scores up to two steps ahead of the values; a place is free
    once its chunk's values, or of a chunk without values its scores (`early`), are multiplied.  Scores come as early as they
    may, values as late, and the warps run as far as their waits let them: the chunks copied into a place still in use."""
    phase = [0] * slots
    lots = [[g for s in range(steps) for g in range(s * chunks + a, s * chunks + min(b, chunks))] for a, b in ((0, 2), (2, 4))]
    at, wrong, copied = [0, 0], [], set()

    def run():
        for w in (0, 1):
            while at[w] < len(lots[w]):
                g = lots[w][at[w]]
                turn, place = g // slots, g % slots
                if turn > 0 and phase[place] % 2 == (turn - 1) % 2:
                    break
                if phase[place] < turn:
                    wrong.append(g)
                copied.add(g)
                at[w] += 1

    def free(s, some):
        for c in some:
            phase[(s * chunks + c) % slots] += 1
        run()

    run()
    values = 0
    for s in range(steps):
        if s - values > 1:
            free(values, range(blocks if early else chunks))
            values += 1
        if not all(s * chunks + c in copied for c in range(chunks)):
            return wrong, s
        if early:
            free(s, range(blocks, chunks))
    return wrong, steps


@pytest.mark.parametrize("heads,place", [(64, 0), (32, 1), (16, 2)])
def test_a_place_of_the_ring_is_free_before_it_is_copied_to(heads, place):
    src = code("attend_cache8.cu")
    slots = [int(x) for x in re.search(r"int slots_of\(int heads\) \{ return heads == 64 \? (\d+) : heads == 32 \? (\d+) : (\d+); \}", src).groups()]
    scores = src[src.index("auto scores = "):src.index("auto values = ")]
    early = "kv_free" in scores
    for chunks in (1, 2, 3, 4):
        for blocks in range(1, chunks + 1):
            wrong, steps = ring(slots[place], chunks, blocks, early)
            assert not wrong and steps == 60, (heads, chunks, blocks, wrong[:5], steps)
