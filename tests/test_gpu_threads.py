"""Calls of several host threads at once, each with its own stream, workspace and outputs."""
import ctypes
import threading

import pytest
import torch

from mixture_experts_layer_29_b200 import abi, norm

pytestmark = pytest.mark.gpu


def test_norm_gradients_of_two_shapes_from_several_threads(cuda_device):
    """The gradients of a wide and of a narrow row share a kernel and need different amounts of shared
    memory: no thread's call may meet another's."""
    T, widths, calls = 4, (6144, 768) * 3, 5000
    L, errors, start = norm.lib(), [], threading.Barrier(len(widths))

    def work(H):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            g = torch.Generator(device="cuda").manual_seed(H)
            rows = lambda: torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)     # noqa: E731
            d = norm.make_desc(T, H)
            dr, dn, r, b = rows(), rows(), rows(), rows()
            w, rstd = torch.ones(H, device="cuda"), torch.ones(T, device="cuda")
            out = [torch.empty_like(b), torch.empty_like(b), torch.empty_like(w), torch.empty_like(w)]
            ws = norm.workspace(d)
            norm.block_norm_backward(d, dr, dn, r, b, w, None, w, rstd, rstd, out[0], out[1], out[2], None, out[3], ws)
            want = [t.clone() for t in out]
            for t in out:
                t.zero_()
            # the C call itself, so that the threads spend their time there
            p = [t if t is None else t.data_ptr() for t in
                 (dr, dn, r, b, w, None, w, rstd, rstd, out[0], out[1], out[2], None, out[3], ws)]
            desc, n = ctypes.byref(d), ws.numel()
            st.synchronize()
            start.wait()
            codes = {L.moe_block_norm_backward(desc, *p, n, st.cuda_stream) for _ in range(calls)}
            st.synchronize()
            if codes != {0} or not all(torch.equal(x, y) for x, y in zip(out, want)):
                errors.append((H, codes))

    threads = [threading.Thread(target=work, args=(H,)) for H in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_permutations_of_two_layers_from_several_threads(cuda_device):
    """Layers of different numbers of experts share the small batches' kernel, not its shared memory."""
    T, n_ffn, K, H, calls = 512, (1000, 400), 4, 128, 3000
    L, errors, start = abi.lib(), [], threading.Barrier(6)

    def work(n):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            b = abi.StepBuffers.allocate(abi.make_shape(T, H, 128, n, 0, K, "bf16", "deterministic"))
            g = torch.Generator(device="cuda").manual_seed(n)
            idx = torch.rand(T, n, device="cuda", generator=g).argsort(1)[:, :K].int().contiguous()
            gate = torch.ones(T, K, device="cuda")
            b.zgate.zero_()
            x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
            args = (b.shape, idx, gate, b.zgate, x, b.offsets, b.perm_token, b.row_of, b.row_gate, b.x_perm, None, b.ws)
            abi.permute(*args)
            want = b.row_of.clone()
            b.row_of.fill_(-9)
            p = [None if t is None else t.data_ptr() for t in args[1:]]
            shape, ws = ctypes.byref(b.shape), b.ws.numel()
            st.synchronize()
            start.wait()
            codes = {L.moe_permute(shape, *p, ws, st.cuda_stream) for _ in range(calls)}
            st.synchronize()
            if codes != {0} or not torch.equal(b.row_of, want):
                errors.append((n, codes))

    threads = [threading.Thread(target=work, args=(n,)) for n in n_ffn * 3]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
