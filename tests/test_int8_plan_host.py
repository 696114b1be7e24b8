"""The form and the workspace of moe_int8_product by sizes (no GPU): csrc/int8_plan.cuh
compiled for the host, and the library's workspace size beside it."""

import pytest

from _int8_plan import CASES, X, form, plans

import mixture_experts_ffn_14_b200 as moe


def test_forms_at_the_grok_shape():
    d, f, E = 6144, 32768, 8
    for m, up, down in ((16, ("stream", 64), ("stream", 64)), (48, ("stream", 64), ("stream", 64)),
                        (128, ("stream", 128), ("stream", 128)), (192, ("pair", 256), ("pair", 256)),
                        (256, ("pair", 512), ("pair", 256)), (287, ("pair", 512), ("pair", 512)),
                        (525, ("pair", 512), ("pair", 256)), (1024, ("pair", 512), ("pair", 512))):
        assert form(E * m, d, f, E, pair=True)[:2] == up, m
        assert form(E * m, f, d, E)[:2] == down, m
    # one row more than a form's last
    assert form(E * 48 + 1, d, f, E, pair=True)[:2] == ("stream", 128)
    assert form(E * 128 + 1, d, f, E, pair=True)[0] == "pair"


def test_split_form_by_tiles_and_k_blocks():
    def split(tiles, blocks, R=16):
        got = form(R, 128 * blocks, 256 * tiles)
        assert got[0] == ("split" if got[2] else "stream")
        return got[2]

    last = {8: 14, 6: 21, 5: 25, 4: 32, 3: 44, 2: 73}   # tiles that clusters of that many CTAs run in one wave
    for (s, tiles), (after, _) in zip(last.items(), list(last.items())[1:] + [(0, 0)]):
        assert split(tiles, 40) == s and split(tiles + 1, 40) == after
    assert split(14, 16) == 8 and split(14, 15) == 6    # two K blocks for each CTA at least
    assert split(10, 4) == 2 and split(10, 3) == 0
    assert split(11, 192) == 8 and split(11, 193) == 0  # few CTAs with long runs
    assert split(12, 300) == 8
    # an expert's last tile may be short: one more tile for each expert but one
    assert form(16, 4096, 256, 8) == ("split", 64, 8) and form(16, 4096, 512, 8) == ("split", 64, 6)


def test_the_products_of_the_gpu_tests_take_the_forms_they_are_meant_for():
    for name, tile, R, K, N, rows, pair in CASES:
        assert sum(rows) <= R
        for x in X:
            assert form(R, K, N, len(rows), x, pair)[:2] == (name, tile), (name, tile, R, K, N)
        if tile == 512:
            assert sum(-(-m // 512) for m in rows) * -(-N // (128 if pair else 256)) > 2 * 74
            assert any(0 < m % 512 <= 256 for m in rows)
    assert {(c[0], c[1]) for c in CASES} == {("split", 64), ("split", 128), ("stream", 64), ("stream", 128),
                                             ("pair", 256), ("pair", 512)}


@pytest.mark.parametrize("x", list(X))
@pytest.mark.parametrize("pair", [False, True])
def test_workspace_size_is_the_plans(x, pair):
    sizes = [(c[2], c[3], c[4], len(c[5]), x, pair) for c in CASES]
    sizes += [(1, 16, 16, 1, x, pair), (1 << 24, 16, 16, 1024, x, pair), (5, 131056, 1 << 20, 3, x, pair)]
    for s, (_, _, _, ws) in zip(sizes, plans(sizes)):
        assert moe.moe_int8_workspace_size(s[0], s[1], s[2], s[3], X[x], pair) == ws
