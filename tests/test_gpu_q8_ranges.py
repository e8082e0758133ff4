"""The 8-bit cache's calls at the ends of their ranges: as many indices as 32 bits
count, forms that only long prompts take, values far apart, rows that one key
rules over a long cache."""
import numpy as np
import pytest
import torch

from q8_helpers import BF16, f64, i32
from ranking_prefill_gb300 import lib
from test_gpu_q8_rows import Cache, check_exact, draw, ws

pytestmark = pytest.mark.gpu


def test_as_many_indices_as_32_bits_count():
    """2^31 - 1 rows by index, most of them skipped: the look at the indices ends, and it sees the last ones."""
    n = 2 ** 31 - 1
    x = draw(np.random.default_rng(1), 3, 4, 128)
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    rows = torch.zeros(n, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 2 ** 30, n - 2049, n - 2, n - 1], device="cuda")
    src = [0, 1, 2, 1, 2]
    slots[at] = i32([5, 6, 7, 8, 9])
    rows[at] = i32(src)
    ca, s = Cache(1, 16, 4, 128), ws()
    lib.mis_paged_write_kv_q8(ca.c, x.cuda(), x.cuda(), slots, s, src_rows=rows)
    assert lib.mis_get_device_status(s) == lib.MIS_OK
    kc, ke, vc, ve = ca.rows()
    for c, e in ((kc, ke), (vc, ve)):
        check_exact(c[5:10], e[5:10], f64(x)[src])
        assert (c[:5] == 0x55).all() and (c[10:] == 0x55).all() and (e[:5] == 0x66).all()
    for bad, where in ((16, slots), (3, rows)):
        was = where[n - 1].clone()
        where[n - 1] = bad
        lib.mis_paged_write_kv_q8(ca.c, x.cuda(), x.cuda(), slots, s, src_rows=rows)
        assert lib.mis_get_device_status(s) == lib.MIS_ERR_DEVICE_INDEX
        where[n - 1] = was
