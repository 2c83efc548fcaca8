"""Host logic of the attention's choice of kernels (i8_kv_attend_config, no GPU)."""
import itertools

import pytest

import ternary_weight_decode_amd as tw

ANY = 2 ** 31 - 1


def workspace_of(launches, d, nseq):
    """Bytes of a plan: two parts of every workgroup of a line (D sums, a maximum and a sum a column), and where
    each sequence starts in it."""
    return sum(2 * p["groups"] * p["cols"] * (4 * d + 8) + (nseq + 4) // 4 * 16 for p in launches if p["groups"])


@pytest.mark.parametrize("hq, heads, d", [(32, 8, 128), (16, 8, 128), (1, 1, 64), (20, 1, 128)])
def test_plan_invariants(hq, heads, d):
    g = hq // heads
    for tokens, nseq, width, window, max_rows in itertools.product(
            (1, 7, 64, 500, 5000), (1, 2, 70), (0, 1, 30, 700), (0, 1, 500), (0, 16, 5000)):
        max_len = max(1, 64 * width)
        launches = tw.i8_kv_attend_config(tokens, hq, heads, d, nseq, width, window, max_len, max_rows)
        where = (tokens, nseq, width, window, max_rows, launches)
        assert len(launches) in (1, 2), where
        for p in launches:
            assert p["cols"] in (16, 32, 64, 256) and (not p["streams"] or p["cols"] == 16), where
            tiles = tokens * g // p["cols"] + nseq
            assert p["grid"] == (p["groups"] or tiles * heads), where
        # every count of columns is some launch's, and one's only
        ranges = sorted((p["min_cols"], p["max_cols"]) for p in launches)
        assert ranges[0][0] == 0 and ranges[-1][1] == ANY, where
        assert all(a[1] + 1 == b[0] for a, b in zip(ranges, ranges[1:])), where
        need = tw.i8_kv_attend_workspace_bytes(tokens, hq, heads, d, nseq, max_len, max_rows)
        used = workspace_of(launches, d, nseq)
        assert used == need if window == 0 else used <= need, where


def test_a_line_past_32_bits_is_not_taken():
    wide = 2 ** 31 // 64 - 1
    assert tw.i8_kv_attend_config(1, 32, 8, 128, 1, 1000)[0]["groups"] > 0
    assert tw.i8_kv_attend_config(1, 32, 8, 128, 1, wide)[0]["groups"] > 0
    assert tw.i8_kv_attend_config(64, 32, 8, 128, 64, wide, max_len=50000)[0]["groups"] == 0


def test_plan_arguments():
    args = dict(tokens=1, hq=4, heads=2, d=128, nseq=1, width=4)
    for bad in (dict(d=96), dict(hq=3), dict(hq=0), dict(tokens=-1), dict(nseq=-1), dict(width=-1), dict(window=-1),
                dict(max_len=0), dict(max_rows=-1), dict(width=2 ** 31 // 64)):
        with pytest.raises(RuntimeError):
            tw.i8_kv_attend_config(**{**args, **bad})
    assert tw.i8_kv_attend_config(**{**args, "tokens": 0}) == tw.i8_kv_attend_config(**{**args, "nseq": 0}) == []
    assert tw.lib().i8_kv_attend_config(1, 4, 2, 128, 1, 4, 0, 256, 0, None) == -1
