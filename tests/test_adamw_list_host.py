"""The optimiser's list of tensors as the library's structure, on the host."""
import ctypes

from transformer_xl_relative_rel_gb300 import abi


def test_packed_fields_lie_where_the_structure_has_them():
    fields, entry = abi._AdamwTensor._fields_, ctypes.sizeof(abi._AdamwTensor)
    values = [0x100 + k for k in range(8)] + [0.5, 1, 0]
    array = (abi._AdamwTensor * 3)()
    assert abi._ADAMW_FIELDS.size <= entry and len(fields) == len(values)
    abi._ADAMW_FIELDS.pack_into(array, entry, *values)
    assert [getattr(array[1], name) for name, _ in fields] == values
    abi._ADAMW_FIELDS.pack_into(array, entry, *[0] * 8, float("inf"), 0, 1)
    assert array[1].param is None and array[1].weight_decay == float("inf") and array[1].grad_dtype == 1
    for k in (0, 2):
        assert not any(bytes(array)[k * entry:(k + 1) * entry])
