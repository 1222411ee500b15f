"""Refusals of the paged serving step's entry points (host checks, no GPU), and
the plain plan itself on hand-made steps."""
import ctypes

import pytest
import torch

from tests import paged_ref as R

FAKE = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def g():
    from routed_head_gqa_b200 import build as gqe_build

    gqe_build.build()
    import routed_head_gqa_b200 as g

    return g


PLAN = dict(n_seqs=4, rows=8, page_size=16, num_pages=32, max_blocks=8, lengths=FAKE, new_lens=FAKE, free_pages=FAKE,
            free_count=FAKE, block_table=FAKE, lengths_out=FAKE, free_count_out=FAKE, cu_new=FAKE, slots=FAKE,
            workspace=FAKE, workspace_bytes=256)


@pytest.mark.parametrize("change,code", [
    (dict(n_seqs=0), 1), (dict(rows=-1), 1), (dict(num_pages=0), 1), (dict(max_blocks=0), 1),
    (dict(page_size=0), 1), (dict(page_size=24), 1), (dict(page_size=1 << 17), 1),
    *[({name: None}, 1) for name in ("lengths", "new_lens", "free_pages", "free_count", "block_table", "lengths_out",
                                     "free_count_out", "cu_new", "slots", "workspace")],
    (dict(workspace=FAKE + 16), 1), (dict(workspace_bytes=255), 1),
    (dict(n_seqs=16385), 2), (dict(page_size=1 << 16, num_pages=1 << 15), 2), (dict(page_size=1 << 16, max_blocks=1 << 15), 2),
])
def test_plan_refuses(g, change, code):
    assert g._lib.gqe_page_plan(*{**PLAN, **change}.values(), None) == code


@pytest.mark.parametrize("change", [dict(lengths_out=FAKE), dict(lengths_out=FAKE + 12), dict(lengths=FAKE + 0x1000 + 12),
                                    dict(free_count_out=FAKE)])
def test_plan_refuses_state_in_place(g, change):
    """The state after the step in the memory of the state before it."""
    apart = dict(lengths_out=FAKE + 0x1000, free_count_out=FAKE + 0x2000)
    assert g._lib.gqe_page_plan(*{**PLAN, **apart, **change}.values(), None) == 1


@pytest.mark.parametrize("change,code", [
    *[({name: None}, 1) for name in ("K_new", "V_new", "slots", "K_pages", "V_pages", "workspace")],
    (dict(K_new=FAKE + 8), 1), (dict(V_pages=FAKE + 4), 1), (dict(num_pages=0), 1), (dict(page_size=3), 1),
    (dict(k_stride=255), 1), (dict(v_stride=260), 1),  # shorter than a row; not 16-byte steps
    (dict(workspace_bytes=0), 1), (dict(page_size=1 << 16, num_pages=1 << 15), 2),
])
def test_append_refuses(g, change, code):
    s = g.make_shape(1, 8, 64, 8, 2, 128, 1, g.GQE_BF16)
    base = dict(K_new=FAKE, k_stride=256, V_new=FAKE, v_stride=256, slots=FAKE, K_pages=FAKE, V_pages=FAKE, num_pages=4,
                page_size=16, workspace=FAKE, workspace_bytes=256)
    assert g._lib.gqe_kv_append(ctypes.byref(s), *{**base, **change}.values(), None) == code


def test_append_refuses_odd_rows(g):
    s = g.make_shape(1, 8, 64, 1, 1, 3, 1, g.GQE_BF16)  # rows of 6 bytes
    assert g._lib.gqe_kv_append(ctypes.byref(s), FAKE, 8, FAKE, 8, FAKE, FAKE, FAKE, 4, 16, FAKE, 256, None) == 2


ATTN = dict(Q=FAKE, K_pages=FAKE, V_pages=FAKE, num_pages=16, page_size=16, block_table=FAKE, max_blocks=8, n_seqs=2,
            cu_new=FAKE, lengths=FAKE, window=0, sinks=0, idx=FAKE, gate=FAKE, O=FAKE, workspace=FAKE,
            workspace_bytes=1 << 30)


@pytest.mark.parametrize("change,code", [
    *[({name: None}, 1) for name in ("Q", "K_pages", "V_pages", "block_table", "cu_new", "lengths", "idx", "gate", "O",
                                     "workspace")],
    (dict(Q=FAKE + 2), 1), (dict(K_pages=FAKE + 8), 1), (dict(O=FAKE + 8), 1),
    (dict(num_pages=0), 1), (dict(max_blocks=0), 1), (dict(n_seqs=0), 1), (dict(page_size=12), 1),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(workspace_bytes=256), 1), (dict(workspace=FAKE + 1), 1),
    (dict(page_size=1 << 16, max_blocks=(1 << 14) + 1), 2), (dict(page_size=1 << 16, num_pages=1 << 15), 2),
])
def test_attention_refuses(g, change, code):
    s = g.make_shape(1, 8, 64, 8, 2, 128, 2, g.GQE_BF16)
    assert g._lib.gqe_attn_chunk_paged(ctypes.byref(s), *{**ATTN, **change}.values(), None) == code


def test_attention_refuses_shapes(g):
    call = lambda *a: g._lib.gqe_attn_chunk_paged(ctypes.byref(g.make_shape(*a)), *ATTN.values(), None)  # noqa: E731
    assert call(2, 8, 64, 8, 2, 128, 2, g.GQE_BF16) == 1   # the step is packed: B is 1
    assert call(1, 8, 64, 8, 2, 96, 2, g.GQE_BF16) == 2
    assert call(1, 8, 64, 8, 3, 128, 2, g.GQE_BF16) == 1
    assert call(1, 8, 64, 64, 2, 128, 17, g.GQE_BF16) == 2
    assert call(1, 1 << 23, 64, 256, 2, 32, 2, g.GQE_BF16) == 2  # T * h of 2^31
    assert call(1, 1 << 23, 64, 256, 2, 32, 2, g.GQE_F32) == 2
    assert g.gqe_chunk_workspace_bytes(g.make_shape(1, 8, 64, 8, 3, 128, 2, g.GQE_BF16)) == 0


def test_binding_refuses_host_tensors(g):
    """Tensors that are not on the current GPU are refused before any pointer is passed on."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(g.GQEError, match="INVALID_ARGUMENT"):
        g.gqe_page_plan(16, i(2), i(2), i(8), i(1), i(2, 4), i(2), i(1), i(3), i(5), ws)
    s = g.make_shape(1, 5, 64, 8, 2, 128, 1, g.GQE_BF16)
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(g.GQEError, match="INVALID_ARGUMENT"):
        g.gqe_kv_append(s, b(5, 2, 128), b(5, 2, 128), i(5), b(4, 16, 2, 128), b(4, 16, 2, 128), ws)
    with pytest.raises(g.GQEError, match="INVALID_ARGUMENT"):
        g.gqe_attn_chunk_paged(s, b(5, 8, 128), b(4, 16, 2, 128), b(4, 16, 2, 128), i(2, 4), i(3), i(2), 0, 0,
                               i(5, 2, 1), torch.zeros(5, 2, 1), b(5, 8, 128), ws)


def test_status_names(g):
    assert g.gqe_status_string(g.GQE_ERR_OUT_OF_PAGES) == "GQE_ERR_OUT_OF_PAGES"


def test_plain_plan_by_hand():
    """Pages of 4 rows: request 0 ends (2 pages back), 1 stays in its page, 2 grows by two pages, 3 starts."""
    table = [[5, 6, -1], [7, -1, -1], [8, -1, -1], [-1, -1, -1]]
    out, free, cu, slots, pushed = R.plan(4, 12, 3, 14, [6, 2, 4, 0], [-1, 1, 6, 5], [1, 2, 3], table)
    assert pushed == [5, 6]
    assert out == [0, 3, 10, 5] and cu == [0, 0, 1, 7, 12]
    assert table == [[5, 6, -1], [7, -1, -1], [8, 6, 5], [3, 2, -1]] and free == [1]
    assert slots == [30, 24, 25, 26, 27, 20, 21, 12, 13, 14, 15, 8, -1, -1]
    with pytest.raises(R.Refused, match="pages"):
        R.plan(4, 12, 3, 14, [0], [9], [1, 2], [[-1, -1, -1]])
    for bad in ([-1], [13]):
        with pytest.raises(R.Refused, match="arguments"):
            R.plan(4, 12, 3, 14, bad, [0], [1, 2], [[-1, -1, -1]])
