"""Calls on a stream that is not the current one, with no workspace given: theirs is the call's for as long as it runs."""
import pytest
import torch

import tree_speculative_decoding_array_gb300 as tsv

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def calls():
    rows, H, V, k = 24, 512, 30011, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    n = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    f32 = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
    x, W, hidden = n(rows, V), n(V, H).half(), n(rows, H).bfloat16()
    W8, ws = n(V, H).to(F8), 0.01 + torch.rand(-(-V // 128), H // 128, device=DEV, generator=g)
    a, sa = torch.empty(rows, H, dtype=F8, device=DEV), f32(rows, H // 128)
    tsv.quantize_e4m3(hidden, a, sa)
    u = torch.rand(rows, device=DEV, generator=g)
    top, lp, tok = i32(rows, k), f32(rows, k), i32(rows)
    return dict(
        draft_children=(tsv.load().tsv_draft_children_workspace_size(rows, V, k), (top, lp),
                        lambda st: tsv.draft_children(x, top, lp, top_k=k, stream=st)),
        token_logprobs=(tsv.token_logprobs_workspace_size(rows, V, k), (top, lp),
                        lambda st: tsv.token_logprobs(x, top_tokens=top, top_logp=lp, stream=st)),
        matmul_e4m3_argmax=(256, (tok,), lambda st: tsv.matmul_e4m3_argmax(a, sa, W8, ws, tok, stream=st)),
        lm_head_argmax=(tsv.lm_head_workspace_size(rows, H, V, tsv.F16), (tok,),
                        lambda st: tsv.lm_head_argmax(hidden, W, tok, w_dtype=tsv.F16, V=V, stream=st)),
        lm_head_logits=(tsv.lm_head_workspace_size(rows, H, V, tsv.E4M3_B128), (x,),
                        lambda st: tsv.lm_head_logits(hidden, W8, x, w_dtype=tsv.E4M3_B128, V=V, scales=ws, stream=st)),
        sample_nucleus=(tsv.sample_workspace_size(rows, V, 20), (tok,),
                        lambda st: tsv.sample_nucleus(x, u, tok, temperature=1.0, top_k=20, top_p=0.9, stream=st)))


@pytest.mark.parametrize("name", ["draft_children", "token_logprobs", "matmul_e4m3_argmax", "lm_head_argmax", "lm_head_logits", "sample_nucleus"])
def test_the_current_stream_does_not_get_a_workspace_in_use(gpu_lib, name):
    size, outs, call = calls()[name]
    assert size > 0
    call(None)
    bool((torch.full((size,), 0x5A, dtype=torch.uint8, device=DEV) == 0x5A).all())  # a kernel's first use may wait for the GPU
    want = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about 0.1 s: the call's kernels run after everything below has been asked for
    call(side)
    others = [torch.full((size,), 0x5A, dtype=torch.uint8, device=DEV) for _ in range(16)]
    torch.cuda.synchronize()
    assert all(bool((t == 0x5A).all()) for t in others)
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("name", ["token_logprobs", "matmul_e4m3_argmax", "lm_head_argmax"])
def test_a_stream_of_another_kind(gpu_lib, name):
    """A stream made outside of torch, known by its handle alone."""
    _, outs, call = calls()[name]
    call(None)
    want = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    class Handle:
        cuda_stream = side.cuda_stream

    call(Handle())
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_rows_at_any_address_give_the_same_bits_on_another_stream(gpu_lib):
    """The other stream waits for the inputs and for what the outputs were filled with."""
    base = torch.randn(4 * 50001 + 3, device=DEV)
    x = base[3:].view(4, 50001)
    targets = torch.tensor([0, 1, 2, 50000], dtype=torch.int32, device=DEV)

    def ask(stream):
        o = dict(logp=torch.full((4,), 7.5, device=DEV), entropy=torch.full((4,), 7.5, device=DEV), rank=torch.full((4,), -9, dtype=torch.int32, device=DEV),
                 top_tokens=torch.full((4, 20), -9, dtype=torch.int32, device=DEV), top_logp=torch.full((4, 20), 7.5, device=DEV))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        tsv.token_logprobs(x, targets, stream=stream, **o)
        torch.cuda.synchronize()
        return o

    one, two = ask(None), ask(torch.cuda.Stream())
    assert all(torch.equal(one[n], two[n]) for n in one)
