"""The cache calls' binding: what is missing is named, how attention's work is
dealt out shows in its workspace, and the package imports on a PyTorch build
without GPU support."""

import os
import subprocess
import sys

import pytest
import torch

mq = pytest.importorskip("mqa_logits_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


CALLS = {
    mq.paged_kv_slots: dict(context_lens=i32(2), new_lens=i32(2), free_blocks=i32(3), block_table=i32(2, 4),
                            num_blocks=9, block_size=16, max_context_len=16, max_tokens=4),
    mq.paged_kv_write: dict(fmt="mxfp4", x=torch.zeros(2, 2, 64), slots=torch.zeros(2, dtype=torch.int64),
                            kv_pool=u8(3, 16, 2, 32), kv_sf_pool=u8(3, 16, 2, 2)),
    mq.paged_attention: dict(fmt="mxfp4", q=torch.zeros(2, 4, 64, dtype=torch.bfloat16), k_pool=u8(3, 16, 2, 32),
                             k_sf_pool=u8(3, 16, 2, 2), v_pool=u8(3, 16, 2, 32), v_sf_pool=u8(3, 16, 2, 2),
                             context_lens=i32(2), block_table=i32(2, 4), next_n=1, max_context_len=16),
}
TENSORS = [(fn, name) for fn, args in CALLS.items() for name, x in args.items() if isinstance(x, torch.Tensor)]


@pytest.mark.parametrize("fn,name", TENSORS, ids=lambda x: x if isinstance(x, str) else x.__name__)
def test_what_is_missing_is_named(fn, name):
    with pytest.raises(ValueError, match=name + " is required"):
        fn(**{**CALLS[fn], name: None})


@pytest.mark.parametrize("fn,name", TENSORS, ids=lambda x: x if isinstance(x, str) else x.__name__)
def test_scalars_are_refused(fn, name):
    given = CALLS[fn][name]
    with pytest.raises(ValueError):
        fn(**{**CALLS[fn], name: given.new_zeros(())})


@pytest.mark.gpu
@pytest.mark.parametrize("fn,name", TENSORS, ids=lambda x: x if isinstance(x, str) else x.__name__)
def test_what_is_missing_is_named_on_the_gpu(fn, name):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    args = {k: x.cuda() if isinstance(x, torch.Tensor) else x for k, x in CALLS[fn].items()}
    with pytest.raises(ValueError, match=name + " is required"):
        fn(**{**args, name: None})
    with pytest.raises(ValueError):
        fn(**{**args, name: args[name].new_zeros(())})


def test_selected_columns_keep_their_workers():
    # Units of one size are dealt out whole, with nothing to join (no workspace),
    # only where that leaves few of the 512 workers idle: not 257 of them for 514.
    size = mq.paged_attention_workspace_size
    for units, whole in ((512, True), (513, False), (514, False), (520, False), (640, False),
                         (768, False), (1000, True), (1024, True), (1536, True)):
        assert (size(units, 1, 16, 1, 128, 8192, 2048) == 0) == whole, units
    for units, whole in ((256, True), (258, False), (320, False), (500, True), (512, True)):
        assert (size(units, 1, 64, 1, 128, 8192, 2048) == 0) == whole, units


def test_imports_without_gpu_support_in_torch():
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_get')]:\n"
            "    delattr(torch._C, name)\n"
            "import mqa_logits_amd\n"
            "assert mqa_logits_amd.paged_attention_workspace_size(1, 1, 8, 1, 128, 100000) > 0\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
