"""Results of nk_verify_drafts over what it reads are refused before anything is launched (CPU only): every block of a sequence
reads the drafts and their counts while one of them writes the results."""
import pytest

import quantized_paged_kv_cache_gb300 as nk

# fake buffers, far apart; never dereferenced: every call below fails host validation
BUF = {n: (i + 1) << 24 for i, n in enumerate(("p", "q", "d", "n", "u", "ctx", "tokens", "acc", "nxt"))}
B, T, V = 3, 3, 100
BYTES = dict(p=B * T * V * 4, q=B * (T - 1) * V * 4, d=B * (T - 1) * 4, n=B * 4, u=B * T * 4, ctx=B * 4, tokens=B * T * 4, acc=B * 4,
             nxt=B * 4)


def call(**at):
    a = BUF | at
    return nk.lib().nk_verify_drafts(a["p"], V, a["q"], V, a["d"], a["n"], a["u"], B, T, V, a["ctx"], a["tokens"], a["acc"], a["nxt"], None,
                                     None)


@pytest.mark.parametrize("result", ["tokens", "acc", "nxt"])
@pytest.mark.parametrize("other", ["p", "q", "d", "n", "u", "ctx"])
def test_results_over_inputs(result, other):
    if (result, other) != ("nxt", "ctx"):  # (these two may be one buffer)
        assert call(**{result: BUF[other]}) == 2
    assert call(**{result: BUF[other] + BYTES[other] - 4}) == 2  # its first entry over the last one
    assert call(**{result: BUF[other] - BYTES[result] + 4}) == 2


@pytest.mark.parametrize("one,two", [("tokens", "acc"), ("tokens", "nxt"), ("acc", "nxt")])
def test_results_over_each_other(one, two):
    assert call(**{one: BUF[two]}) == 2
    assert call(**{two: BUF[one] + BYTES[one] - 4}) == 2


def test_rows_apart():
    """Rows further apart than the vocabulary: the last row's end counts, not the last stride's."""
    args = [BUF["p"], 1 << 20, BUF["q"], 1 << 20, BUF["d"], None, BUF["u"], B, T, V, None]
    end = BUF["p"] + ((B * T - 1) * (1 << 20) + V) * 4
    assert nk.lib().nk_verify_drafts(*args, end - 4, BUF["acc"], None, None, None) == 2
