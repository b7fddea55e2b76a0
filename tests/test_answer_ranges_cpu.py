"""Ranges of the calls at the answering end that are refused on the host."""
import pytest

import rank_delta_gb300 as rd
from rank_delta_gb300 import build as rdbuild
from tests.test_abi_cpu import expect


@pytest.fixture(scope="module", autouse=True)
def built():
    rdbuild.build()
    return rd.lib()


@pytest.mark.parametrize("inv_t", [1.001 * 2.0 ** 127, 2.5e38, 3.4e38])
def test_inverse_temperatures_that_the_arithmetic_does_not_take(inv_t):
    """Times log2 e some of them are infinite in fp32, and the largest logit minus itself times that a NaN."""
    expect(rd.LORA_ERR_RANGE, lambda: rd.lora_logprobs(4096, rd.LORA_DTYPE_F32, 100, 0, 100, 256, inv_t, 0, 256, 256, 256, 0, 0, 512, 256),
           contains=("inv_temperature",))
    expect(rd.LORA_ERR_RANGE, lambda: rd.lora_logprobs_grad(4096, rd.LORA_DTYPE_F32, 100, 0, 100, 256, inv_t, 256, 256, 256, 256, 8192,
                                                            100), contains=("inv_temperature",))


def test_projections_of_more_rows_than_a_launch_takes():
    from tests.test_abi_cpu import fake_route
    rt = fake_route(L=4, R=8, K=256, N=256)
    expect(rd.LORA_ERR_UNSUPPORTED, lambda: rd.lora_mx4_proj_apply(4096, 256, 8192, 513, 65535 * 256 + 1, 256, 256, 4096, rt, 4096, 256,
                                                                   1 << 20, 1 << 62), contains=("16776961",))
