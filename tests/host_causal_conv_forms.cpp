// The rows of a strip of the causal convolution (causal_conv_forms.hpp) for tests/test_causal_conv_forms.py.
#include "../quantized_state_space_amd/csrc/causal_conv_forms.hpp"

extern "C" int64_t host_strip(int64_t tokens, int64_t cblocks) { return qssm_conv::strip_rows(tokens, cblocks); }
