// The choice of the block-scaled e4m3 linear layer's tile form (gemm_f8_forms.hpp) for tests/test_gemm_f8_forms.py.
#include "../quantized_state_space_amd/csrc/gemm_f8_forms.hpp"

extern "C" int host_form(int64_t M, int64_t N, int64_t K, int yf16) { return qssm_f8::choose_form(M, N, K, yf16 != 0); }
