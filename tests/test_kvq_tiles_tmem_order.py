"""Loads and stores of tensor memory in the softmax over codes (kv_tiles.cu), on the CPU, from the source: tcgen05.st is
asynchronous, so what it wrote may be loaded again only behind a tcgen05.wait::st. A tile's scores and V's exponent may
each move a row's reference, so that O is loaded, multiplied and stored up to three times to a tile, and P once more."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "attention_fa_fwd_02_gb300", "csrc", "kv_tiles.cu")
CALL = re.compile(r"\b(rescale|tmem_ld32x4|tmem_ld32x2|tmem_ld32|tmem_ld16|tmem_st32|tmem_st16|tmem_st_wait)\(([^;]*?)\)?;")


def block(text, at):
    """What stands between the braces of which the first opens at or after `at`."""
    first = at = text.index("{", at)
    depth = 0
    while True:
        depth += {"{": 1, "}": -1}.get(text[at], 0)
        at += 1
        if depth == 0:
            return text[first + 1:at - 1]


def accesses(text):
    """(call, "o" or "s": the columns it names) in the order of the text."""
    text = re.sub(r"//[^\n]*", "", text)
    return [(m[1], "o" if "o_addr" in m[2] else "s") for m in CALL.finditer(text)]


def unordered(calls):
    """Loads of columns that a store before them may still be on its way to."""
    pending, bad = set(), []
    for i, (what, where) in enumerate(calls):
        if what == "tmem_st_wait":
            pending.clear()
        elif what.startswith("tmem_st"):
            pending.add(where)
        elif where in pending:
            bad.append((i, what, where))
    return bad


def softmax_over_codes():
    """The accesses of one tile, every branch taken: the exponent's move, twice the loop over 64 keys, what follows it."""
    with open(SOURCE) as f:
        text = f.read()
    tile = block(text, text.index("if constexpr (BITS != 0)", text.index("// ------------------------------------------------------------ softmax")))
    name = re.search(r"auto rescale = ", tile).start()
    body = block(tile, tile.index("{", tile.index(")", name)))
    rest = tile.replace(body, "", 1)
    loop = block(rest, rest.index("for (int h = 0; h < 2; ++h)"))
    before, after = rest.split(loop)
    moves = accesses(body)
    assert moves and {c for c, _ in moves} >= {"tmem_ld32", "tmem_st32"}
    out = []
    for call in accesses(before) + 2 * accesses(loop) + accesses(after.split("} else {")[0]):
        out += moves if call[0] == "rescale" else [call]
    assert sum(c == ("tmem_ld32", "o") for c in out) >= 3 and sum(c == ("tmem_st32", "s") for c in out) >= 4
    return out


def test_the_check_tells_a_missing_wait():
    st, ld, wait = ("tmem_st32", "o"), ("tmem_ld32", "o"), ("tmem_st_wait", "s")
    assert unordered([ld, st, ld]) == [(2, "tmem_ld32", "o")]
    assert not unordered([ld, st, wait, ld, st]) and not unordered([("tmem_st32", "s"), ld])


def test_no_load_of_o_or_p_passes_a_store():
    calls = softmax_over_codes()
    # (the scores of keys 64 .. 127 lie behind P's columns, which the first half's stores end before)
    calls = [c for c in calls if c[0] != "tmem_ld32x2"]
    assert not unordered(calls)
