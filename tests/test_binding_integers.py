"""What the binding takes for streams and pointers: any int, subclasses included."""
import enum

from structured_activation_sparsity_b200 import _lib as L


class Handle(enum.IntEnum):
    LEGACY = 0
    SIDE = 4096


class Address(int):
    pass


def test_integers_of_any_class():
    assert L._stream(Handle.SIDE) == 4096 and L._stream(Handle.LEGACY) == 0
    assert L._stream(Address(64)) == 64 and L._stream(None) is None
    assert L._ptrs(Address(256), None, 512, Handle.SIDE) == [256, None, 512, 4096]
    assert L._ptr(Address(256)) == 256
