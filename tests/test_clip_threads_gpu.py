"""clip_grad_norm from host threads that share a stream."""
import threading
import time

import pytest
import torch

import linear_recurrence_scan_row_amd as rl
from linear_recurrence_scan_row_amd import rlca, sequence

pytestmark = pytest.mark.gpu


def test_threads_on_one_stream(gpu_device, monkeypatch):
    """A call is several launches, between which the total and the scale lie in
    its workspace: no other call may enqueue on that workspace meanwhile.  Four
    threads on the default stream, each call held up on its way in."""
    real = rlca.lib()
    guard, inside, most = threading.Lock(), {}, [0]

    class Watched:
        def __getattr__(self, name):
            return getattr(real, name)

        def rlca_clip_grad_norm(self, *args):
            workspace = args[5]
            with guard:
                inside[workspace] = inside.get(workspace, 0) + 1
                most[0] = max(most[0], inside[workspace])
            time.sleep(0.005)
            status = real.rlca_clip_grad_norm(*args)
            time.sleep(0.005)
            with guard:
                inside[workspace] -= 1
            return status

    watched = Watched()
    monkeypatch.setattr(sequence, "lib", lambda: watched)
    # over 96 tensors: two launches for the norm, two for the scaling
    grads = [[torch.full((50 + k,), 1.0 + k, device="cuda") for _ in range(100)] for k in range(4)]
    errors, norms = [], [[] for _ in grads]
    outs = [[[torch.empty_like(t) for t in g] for _ in range(4)] for g in grads]
    start = threading.Barrier(len(grads))

    def run(k):
        try:
            start.wait(timeout=60)
            for out in outs[k]:
                norms[k].append(rl.clip_grad_norm(grads[k], 1.0, out=out))
        except Exception as e:
            errors.append(repr(e))

    threads = [threading.Thread(target=run, args=(k,)) for k in range(len(grads))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    torch.cuda.synchronize()
    assert not errors and not any(t.is_alive() for t in threads)
    assert most[0] == 1
    for k, g in enumerate(grads):
        norm = (1.0 + k) * (100 * (50 + k)) ** 0.5
        for n, out in zip(norms[k], outs[k]):
            assert n.item() == pytest.approx(norm, rel=1e-12)
            scaled = torch.cat(out)
            # eps, the scale's and the product's roundings
            assert torch.allclose(scaled, torch.full_like(scaled, (1.0 + k) / norm), rtol=1e-6)
