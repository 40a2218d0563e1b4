"""A 4-bit linear layer (forward only) over the library's C ABI.

``Int4Linear`` is to ``int4_linear`` what ``Int8Linear`` is to ``int8_linear``:
it holds the prepared 4-bit weight and the bias, nothing else, and its forward
is one call.  Its place is a decode step, where the weight's bytes are what a
layer costs; rows are taken 64 at a time.

The prepared bytes do not say what they are (group_size 64 without and 128 with
zero points, 250 and 256 inputs take the same number of them), so the state
dict has the layer's format beside them, and a state of another format is not
loaded.  A state without one (saved before there was any) is taken as it is.
"""

from __future__ import annotations

import torch

from . import serving


class Int4Linear(torch.nn.Module):
    """y = x W^T + b with W in 4-bit codes and group scales; x float16 or
    bfloat16 (the type of the layer it was made from), [..., in_features]."""

    def __init__(self, weight: serving.Int4Weight, bias=None):
        super().__init__()
        self.in_features, self.out_features = weight.in_features, weight.out_features
        self.group_size, self.zeros = weight.group_size, weight.zeros
        self.register_buffer("Wq", weight.Wq)
        self.register_buffer("params", weight.params)
        if bias is not None:
            self.bias = torch.nn.Parameter(bias.detach().clone(), requires_grad=False)
        else:
            self.register_parameter("bias", None)

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, group_size: int = 128,
                    symmetric: bool = True) -> "Int4Linear":
        """The 4-bit layer of a float16 or bfloat16 nn.Linear on a GPU
        (quantized now)."""
        w = serving.int4_prepare_weight(linear.weight.detach().contiguous(), group_size, symmetric)
        return cls(w, linear.bias)

    @property
    def _format(self) -> dict:
        return dict(in_features=self.in_features, out_features=self.out_features,
                    group_size=self.group_size, zeros=bool(self.zeros))

    def get_extra_state(self) -> torch.Tensor:
        return torch.tensor(list(self._format.values()), dtype=torch.int64)

    def set_extra_state(self, state) -> None:
        pass  # compared before anything is loaded

    def _load_from_state_dict(self, state_dict, prefix, local_metadata, strict, missing_keys,
                              unexpected_keys, error_msgs):
        key = prefix + "_extra_state"
        if key in state_dict:
            names, saved = self._format.keys(), state_dict[key].tolist()
            if saved != [int(x) for x in self._format.values()]:
                error_msgs.append(
                    f"{prefix[:-1] or 'Int4Linear'}: the state is of {dict(zip(names, saved))}, "
                    f"the layer of {self._format}")
                return
        super()._load_from_state_dict(state_dict, prefix, local_metadata, strict, missing_keys,
                                      unexpected_keys, error_msgs)
        if key in missing_keys:
            missing_keys.remove(key)

    @property
    def weight4(self) -> serving.Int4Weight:
        return serving.Int4Weight(self.Wq, self.params, self.out_features, self.in_features,
                                  self.group_size, self.zeros)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"last dimension {x.shape[-1]} != in_features {self.in_features}")
        y = serving.int4_linear(x.reshape(-1, self.in_features), self.weight4, self.bias)
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"bias={self.bias is not None}, group_size={self.group_size}, zeros={self.zeros}")


__all__ = ["Int4Linear"]
