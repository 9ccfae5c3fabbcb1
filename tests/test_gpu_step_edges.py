"""GPU tests of the serving step's operators at the edges of what their calls
allow: several host threads, refused requests, bad pages, values that are not
finite, scales that differ widely, and closer bounds on the attention's error."""
import threading

import numpy as np
import pytest
import torch

import dsa_sparse_mla_topk_gb300 as dsa
import oracle
import step_reference as ref
import test_gpu_step_ops as ops

pytestmark = pytest.mark.gpu
I32 = torch.int32
SHAPES = [(16, 64, 16), (64, 512, 64)]
both_shapes = pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dsa_sparse_mla_topk_gb300 import build
    build.build()
    oracle.build()
    dsa.load_library()


# ---- batch_layout ------------------------------------------------------------------


def test_layout_large_batches_from_several_threads():
    """Batches past 48 KB of shared memory, of different sizes, from three threads: the
    kernel's limit is one for all of them."""
    errors = []

    def work(R):
        c, n, held, table, free, pages = ops._layout_case(R, 2, 20, 16, seed=R)
        want, _ = ref.batch_layout(c, n, held, table, free, 0, page_size=16, num_pages=pages, capacity=int(n.sum()))
        args = (ops.i32(c), ops.i32(n), ops.i32(held), torch.from_numpy(table).cuda(), ops.i32(free), ops.i32([0]))
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        try:
            for _ in range(2000):
                lay = dsa.batch_layout(*args, page_size=16, num_pages=pages, capacity=int(n.sum()), stream=stream)
            stream.synchronize()
            for k, v in lay._asdict().items():
                assert np.array_equal(ops.host(v), want[k]), (R, k)
        except Exception as e:  # noqa: BLE001
            errors.append((R, repr(e)))

    threads = [threading.Thread(target=work, args=(R,)) for R in (8192, 4000, 6000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
