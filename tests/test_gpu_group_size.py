"""The size limit of a group: the flat layout of unpacked AdamW moments counts 64 elements to an int32, which binds
those groups alone.  Groups are only created here, over made-up addresses that no call reads."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,accepted", [("NADAM_F24", True), ("ADAN", True), ("ADAMW", False), ("ADAMW_U8", False)])
def test_limit_of_the_flat_layout(kind, accepted):
    from memory_lean_optimizer_gb300 import lmopt
    d = lmopt.TensorDesc(w_bf16=0x100000, res_u16=None, m=0x200000, v=0x300000, numel=1 << 37, ndim=1)
    d.shape[0] = 1 << 37
    if accepted:
        lmopt.optim_group_destroy(lmopt.optim_group_create([d], getattr(lmopt, f"OPTIM_KIND_{kind}")))
        return
    with pytest.raises(lmopt.LmoptError) as e:
        lmopt.optim_group_create([d], getattr(lmopt, f"OPTIM_KIND_{kind}"))
    assert e.value.code == lmopt.OPTIM_EINVAL
