"""What the binding takes for a pointer and a stream (no CUDA call is made: M = 0 is a no-op)."""
import numpy as np
import pytest

import rank_delta_gb300 as rd
from rank_delta_gb300 import build as rdbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    rdbuild.build()
    return rd.lib()


class Buffer:
    def __init__(self, address):
        self.address = address

    def data_ptr(self):
        return self.address


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("number", [int, np.int64, np.uint64])
def test_pointers_and_streams_may_be_any_integer(number):
    for pointer in (number(4096), Buffer(number(4096))):
        for stream in (None, number(0), Stream(number(0))):
            rd.lora_logprobs(pointer, rd.LORA_DTYPE_F32, 8, 0, 8, pointer, 1.0, 0, None, None, None, None, None, pointer, 256, stream)
            rd.lora_mx4_quantize(pointer, rd.LORA_DTYPE_F32, 32, 0, 32, pointer, pointer, stream)
