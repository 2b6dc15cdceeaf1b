"""Overlapping arguments and sizes past the limits, refused on the host (no GPU)."""

import ctypes

from test_tree_host import _cdesc, lib  # noqa: F401  (lib is a fixture)


def at(n):
    return ctypes.c_void_p(4096 * n)


def inside(n, byte):
    return ctypes.c_void_p(4096 * n + byte)


def test_commit_path_refuses_results_over_its_inputs(lib):  # noqa: F811
    """new_lens is written while other layers' blocks still read the inputs: batch 3, 4 nodes, 5 table columns."""
    d = _cdesc(batch=3, max_blocks_per_seq=5)

    def call(table=at(3), ctx=at(4), path=at(5), m=at(6), new=at(7)):
        return lib.spec_cache_commit_path(at(1), at(2), table, ctx, path, m, new, 4, ctypes.byref(d), None, None)

    for name, size in (("table", 60), ("ctx", 12), ("path", 48), ("m", 12)):
        for byte in (0, 4, size - 4):
            assert call(**{name: at(8), "new": inside(8, byte)}) == -1, (name, byte)
        assert call(**{name: inside(8, 8), "new": at(8)}) == -1, name  # the result's last word


def test_tree_accept_refuses_results_over_its_inputs(lib):  # noqa: F811
    def call(tokens=at(2), par=at(3), mode=at(4), temp=at(5), out=at(6), path=at(7), m=at(8)):
        return lib.spec_tree_accept(at(1), tokens, par, None, 1, mode, temp, out, path, m, 3, 4, 100, None, None)

    for result in ("out", "path", "m"):
        for name in ("tokens", "par", "mode", "temp"):
            assert call(**{name: at(9), result: at(9)}) == -1, (result, name)
    for a, b in (("out", "path"), ("out", "m"), ("path", "m")):
        assert call(**{a: at(9), b: at(9)}) == -1
    assert call(out=at(9), path=inside(9, 44)) == -1


def test_tables_whose_token_counts_do_not_fit_are_refused(lib):  # noqa: F811
    """ceil(length / block_size) is worked out in 32 bits: max_blocks_per_seq * block_size + block_size - 1 has to fit."""
    most = (1 << 31) - 1
    for page, width, ok in ((3, (most - 2) // 3, True), (3, (most - 2) // 3 + 1, False), (1, 1 << 30, True),
                            (65536, 32766, True), (65536, 32767, True), (65536, 32768, False)):
        size = lib.spec_cache_update_workspace(ctypes.byref(_cdesc(batch=1, block_size=page, max_blocks_per_seq=width)))
        assert (size > 0) == ok, (page, width)


def test_workspace_init_refusals(lib):  # noqa: F811
    assert lib.spec_attention_workspace_init(None, 1 << 20, None) == -4
    assert lib.spec_attention_workspace_init(at(1), 4095, None) == -4
    assert lib.spec_attention_workspace_init(inside(1, 16), 4096, None) == -1


def test_workspaces_on_the_host_need_no_device():
    import speculative_decoding_verification_paged_gb300 as sv
    ws = sv.new_attention_workspace(10000, "cpu")
    assert ws.numel() == 10000 and not bool(ws[: sv.ATTN_COUNTER_BYTES].any())
