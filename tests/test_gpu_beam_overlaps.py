"""token_beam_select refuses an output or a workspace that shares a byte with another
array of the call, and takes arrays that lie next to each other."""
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv

R, W, V, K = 3, 4, 100, 5
I32, F32 = torch.int32, torch.float32
SHAPES = dict(logits=((R * W, V), F32), scores=((R, W), F32), finished=((R, W), I32), weights=((R, W), F32), parents=((R, K), I32),
              tokens=((R, K), I32), new_scores=((R, K), F32))
WRITTEN = ("parents", "tokens", "new_scores", "workspace")


@pytest.mark.gpu
@pytest.mark.parametrize("written", WRITTEN)
def test_overlaps(written):
    need = pkv.token_beam_select_workspace_bytes(R, W, V, K)
    size = {name: 4 * shape[0] * shape[1] for name, (shape, _) in SHAPES.items()}
    size["workspace"] = -(-need // 256) * 256
    step = 2 * size["workspace"]  # multiples of 256
    memory = torch.zeros((len(size) + 2) * step, dtype=torch.uint8, device="cuda")
    at = {name: (i + 1) * step for i, name in enumerate(size)}

    def call(**moved):
        memory.zero_()
        args = {}
        for name in size:
            raw = memory[(first := moved.get(name, at[name])):first + size[name]]
            args[name] = raw if name == "workspace" else raw.view(SHAPES[name][1]).view(SHAPES[name][0])
        args["weights"].fill_(1.0)
        pkv.token_beam_select(**args)

    call()
    for other in size:
        if other == written:
            continue
        grain = 256 if "workspace" in (written, other) else 4
        # the same place, its last bytes, and this one's last bytes on its first ones
        for first in (at[other], at[other] + (size[other] - 1) // grain * grain, at[other] - (size[written] - 1) // grain * grain):
            with pytest.raises(pkv.PkvError, match="EINVAL"):
                call(**{written: first})
        call(**{written: at[other] + -(-size[other] // 256) * 256})
        call(**{written: at[other] - -(-size[written] // 256) * 256})
