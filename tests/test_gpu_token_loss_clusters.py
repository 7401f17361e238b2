"""Rows of logits at the numbers of rows where the forward and the one-pass kernels take clusters of another size."""
import numpy as np
import pytest

from tests.test_gpu_token_loss import binding, check_distill, check_logprobs, make_logits, teacher_lists  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T", [8, 19, 20, 38, 39, 57, 58, 76, 77, 152, 153])
@pytest.mark.parametrize("V,dtype", [(70003, "bf16"), (16384, "f32")])
def test_rows_around_each_border(binding, T, V, dtype):  # noqa: F811
    rng = np.random.default_rng(T)
    l = make_logits(rng, T, V, dtype, 1.0, "normal")
    check_logprobs(binding, l, rng.integers(0, V, T), 7, 1.0)
    ids, values = teacher_lists(rng, l, 20, "twice")
    check_distill(binding, l, ids, values, 1.0, rng.random(T) < 0.7, False)


def test_times_do_not_jump(binding):  # noqa: F811
    """38 and 76 rows took longer than twice as many (clusters that had to wait for a place); now at most a tenth."""
    def us(T):
        l, t = torch.randn(T, 131072, device="cuda").bfloat16(), torch.zeros(T, dtype=torch.int64, device="cuda")
        binding.token_logprobs(l, t)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                binding.token_logprobs(l, t)
        times = []
        for _ in range(7):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    assert us(38) <= 1.1 * us(44) and us(76) <= 1.1 * us(77)
