"""What linrec_bwd refuses by address, on the host: nothing is launched."""
import ctypes

from state_space_model_mamba_amd import recurrence

NAMES = "x g i decay h0 seq cs dy dfin dx dg di dd dh0 ws"


def call(**kw):
    p = {k: 0x100000 * (n + 1) for n, k in enumerate(NAMES.split())}
    p.update({k: p[v] for k, v in kw.items()})
    s = recurrence.make_shape(2, 100, 64, 2, gate="decay")
    args = [ctypes.c_void_p(p[k]) for k in NAMES.split()]
    return recurrence.load_library().linrec_bwd(ctypes.byref(s), *args, ctypes.c_size_t(1 << 40), None)


def test_a_gradient_of_states_in_anothers_place():
    # a sequence's first row writes d_initial_states while its last may still read d_final_states
    assert call(dh0="dfin") == -1
    for k in ("x", "g", "i", "dy"):
        assert call(dx=k) == -1
