"""The absorbed form with more row tiles than half of the GPU's SMs (77 x 64 query rows and more): one run of the whole line a row
tile, no sequence is cut and no scratch is taken."""
import pytest
import torch

from latent_ref import latent_decode_reference, latent_state
from paged_ref import check_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


# (n, nh, dc, dr, page, lens): 4864 rows are two runs on 152 SMs, 4865 one; 10240 are more CTAs than SMs
CASES = [(64, 76, 128, 16, 16, [300, 0, 129]), (61, 80, 128, 16, 64, [40, 500, 3, 0]), (64, 80, 512, 64, 32, [200, 70]),
         (64, 160, 128, 16, 16, [65, 0, 200]), (1, 5003, 256, 32, 16, [0, 100, 250])]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_many_rows(case):
    from bwd_xattn_fwd_gb300 import xattn
    n, nh, dc, dr, page, lens = case
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pages, table = latent_state(len(lens), n, dc + dr, page, lens, seed=n, device="cuda")
    q = (torch.randn(len(lens), n, nh, dc + dr, generator=torch.Generator().manual_seed(nh)) * 0.5).bfloat16().cuda()
    o, lse = xattn.attention_latent_decode(q, pages, i32(table), i32(lens), dc, 0.07)
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    check_tree(o, lse, latent_decode_reference(q, pages, table, lens, dc, 0.07), str(case))


def test_one_run_takes_no_scratch():
    """131072 rows of 512 numbers: as records they would be twice 2056 bytes each, 539 MB that the library's pool would keep."""
    from bwd_xattn_fwd_gb300 import xattn
    n, nh, dc, dr = 64, 2048, 512, 64
    q = torch.zeros(1, n, nh, dc + dr, dtype=torch.bfloat16, device="cuda")
    pages = torch.ones(8, 16, dc + dr, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.arange(8, dtype=torch.int32, device="cuda")[None], torch.tensor([20], dtype=torch.int32, device="cuda")
    o, lse = torch.empty(1, n, nh, dc, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n, nh, device="cuda")

    def call():
        xattn.xattn_latent_decode(q, pages, table, lens, 1, n, nh, dc, dr, 8, 16, 8, 0.1, o, lse,
                                  torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()

    xattn.xattn_trim_scratch(0)
    free = torch.cuda.mem_get_info()[0]
    call()
    assert free - torch.cuda.mem_get_info()[0] < 256 << 20
    assert bool((o == 1).all()) and xattn.xattn_check_device_status() == 0
