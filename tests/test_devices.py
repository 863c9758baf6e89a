"""The calls of a serving step use their tensors' device: tensors of several
devices are refused, and so is a pool of another device than the current one.
No second GPU is needed: the first on tensors without memory, the second on a
made-up CUDA runtime (host_device.cpp)."""
import os
import shutil
import subprocess

import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv
from paged_kv_decode_rope_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def host_program(tmp_path, name):
    """Compile tests/<name>.cpp against the library's internal header and run it."""
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc())))
    exe = str(tmp_path / name)
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-O1", f"-I{build.CSRC}", f"-I{cuda}/include",
                    os.path.join(HERE, name + ".cpp"), "-o", exe], check=True)
    return subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines()


def test_a_pool_of_another_device_is_refused(tmp_path):
    assert host_program(tmp_path, "host_device")[:6] == [
        "pool on 0, current 0: 0", "pool on 0, current 1: -22", "pool on 1, current 0: -22", "pool on 1, current 1: 0",
        "recorded 100", "no device: -5"]


def test_a_kernel_is_set_up_on_every_device(tmp_path):
    assert host_program(tmp_path, "host_device")[6:] == [
        "set-up 0 on 0: 1, set 1 times", "set-up 0 on 1: 1, set 1 times", "set-up 1 on 0: 0, set 2 times",
        "set-up 1 on 1: 0, set 2 times", "set-up 2 on 0: 0, set 2 times", "set-up 2 on 1: 0, set 2 times"]
    # and no kernel keeps that it is set up without the device
    for name in ("logprobs.cu", "prefill.cu", "prefill_scored.cu"):
        with open(os.path.join(build.CSRC, name)) as f:
            text = f.read()
        assert "DeviceSetup" in text and "static std::atomic<bool>" not in text, name


def calls():
    """Every call with the tensors it takes, on meta-like shapes: name -> (function, arguments without their tensors'
    device, the tensors)."""
    i32, f32, bf16, u8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
    return {
        "tables": (pkv.paged_tables_build, {}, dict(
            start_pos=((4,), i32), new_tokens=((4,), i32), free_pages=((9,), i32), free_head=((1,), i32),
            free_head_out=((1,), i32), block_tables=((2, 4, 5), i32), cu_tokens=((5,), i32), seq_lens=((4,), i32),
            positions=((7,), i32), slot_map=((2, 7), i32))),
        "rope": (pkv.paged_rope_append, {}, dict(
            q=((3, 8, 64), bf16), k=((3, 2, 64), bf16), v=((3, 2, 64), bf16), q_rot=((3, 8, 64), f32),
            slot_map=((3,), i32), positions=((3,), i32), rope_table=((4096,), u8))),
        "decode": (pkv.paged_gqa_decode_scored, dict(scale=0.125), dict(
            q_rot=((3, 8, 64), f32), out=((3, 8, 64), f32), block_tables=((3, 5), i32), seq_lens=((3,), i32),
            workspace=((4096,), u8), alibi_slopes=((8,), f32), first_keys=((3,), i32))),
        "prefill": (pkv.paged_gqa_prefill_scored, dict(scale=0.125), dict(
            q_rot=((6, 8, 64), f32), out=((6, 8, 64), f32), block_tables=((3, 5), i32), cu_tokens=((4,), i32),
            start_pos=((3,), i32), workspace=((4096,), u8), alibi_slopes=((8,), f32), prefix_lens=((3,), i32),
            doc_starts=((6,), i32))),
        "logprobs": (pkv.token_logprobs, {}, dict(
            logits=((4, 100), bf16), targets=((4,), i32), logprobs=((4,), f32), entropy=((4,), f32),
            top_ids=((4, 5), i32), top_logprobs=((4, 5), f32), workspace=((4096,), u8)))}


@pytest.mark.skipif(torch.cuda.is_available(), reason="devices that are made up")
@pytest.mark.parametrize("name", ["tables", "rope", "decode", "prefill", "logprobs"])
def test_tensors_of_two_devices_are_refused(name):
    from torch._subclasses.fake_tensor import FakeTensorMode
    function, other, shapes = calls()[name]
    pool = [] if name == "logprobs" else [pkv.KVPool(0, None, 2)]
    with FakeTensorMode():
        for moved in shapes:
            args = {n: torch.empty(s, dtype=t, device="cuda:1" if n == moved else "cuda:0")
                    for n, (s, t) in shapes.items()}
            with pytest.raises(ValueError, match="one device, got cuda"):
                function(*pool, **args, **other)
