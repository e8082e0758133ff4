"""Paged-cache calls on views of one buffer: refused where an output lies over
an input, accepted where rows of one stride lie beside each other."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_paged as T  # noqa: E402
from ranking_prefill_gb300 import lib  # noqa: E402

pytestmark = pytest.mark.gpu


def refused(f, *a, **kw):
    with pytest.raises(lib.MisError) as e:
        f(*a, **kw)
    assert e.value.status == lib.MIS_ERR_INVALID_ARG


def test_views_over_inputs_are_refused():
    t = T.Tree([400], [3], 2, 2, 64, 16, None, seed=60).prepare()
    rows = t.kc.view(-1, 2, 64)
    other = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    ws = T.workspace(256)
    for k, v in ((rows[16:], rows[:-16].clone()), (other, t.vc.view(-1, 2, 64)[100:108])):
        refused(lib.mis_paged_write_kv, t.cache, k, v, T.i32([1, 2]), ws)
    twice = torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    q, k = twice[:3], twice[1:]

    def call(q=t.q, k=t.k, v=t.v, o=t.o, lse=t.lse):
        lib.mis_tree_attention_fwd(t.desc, q, k, v, o, lse, t.d_table, t.d_len, t.d_cu, None, t.ws)
    call()
    refused(call, q=q, o=k)
    refused(call, k=q, o=k)
    refused(call, v=k, o=q)
    refused(call, o=rows[20:23])
    refused(call, o=t.vc.view(-1, 2, 64)[300:303])
    refused(call, lse=t.q.view(torch.float32).view(-1)[4:10].view(2, 3))
    refused(call, lse=t.vc.view(torch.float32).view(-1)[64:70].view(2, 3))
    refused(call, lse=t.o.view(torch.float32).view(-1)[100:106].view(2, 3))
    e = T.Extend([3, 4], [5, 6], 16, 4, 9)
    e.d_pos = e.d_slot
    refused(e.call)
    e = T.Extend([3, 4], [5, 6], 16, 4, 9)
    e.d_cu = e.d_free[:3]
    refused(e.call)


@pytest.mark.parametrize("hq,hkv,D,nodes", [(4, 2, 64, [5, 9]), (8, 2, 128, [70, 3])])
def test_one_buffer_of_q_k_v_and_o(hq, hkv, D, nodes):
    # rows of q, k, v and o side by side in one buffer, as a fused projection leaves them
    t = T.Tree([300, 77], nodes, hq, hkv, D, 32, None, seed=61)
    buf = torch.zeros(t.T, 2 * hq + 2 * hkv, D, dtype=torch.bfloat16, device="cuda")
    q, k, v, o = buf.split([hq, hkv, hkv, hq], 1)
    q.copy_(t.q)
    k.copy_(t.k)
    v.copy_(t.v)
    t.q, t.k, t.v = q, k, v
    t.prepare()
    t.o = o
    t.call()
    assert lib.mis_get_device_status(t.ws) == lib.MIS_OK
    t.compare(t.oracle())


def test_rows_beside_the_cache_in_one_buffer():
    # K, V and the rows to store as columns of one buffer
    rng = np.random.default_rng(0)
    buf = torch.zeros(8 * 16, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    kc, vc = buf[:, 0].unflatten(0, (8, 16)), buf[:, 1].unflatten(0, (8, 16))
    buf[:, 2], buf[:, 3] = T.randn(62, 128, 2, 64), T.randn(63, 128, 2, 64)
    T.check_write(kc, vc, buf[:, 2], buf[:, 3], rng.permutation(128)[:100])
