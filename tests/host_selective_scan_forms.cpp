// How the selective scan cuts sequences and places their pieces' ends (selective_scan_forms.hpp) for tests/test_selective_scan_forms.py.
#include "../quantized_state_space_amd/csrc/selective_scan_forms.hpp"

extern "C" int64_t host_piece(int64_t tokens, int64_t nseq, int64_t waves, int packed) {
  return qssm_sscan::piece_rows(tokens, nseq, waves, packed != 0);
}
extern "C" int64_t host_four(int64_t nseq, int64_t blocks, int npl) { return qssm_sscan::four_at_a_time(nseq, blocks, npl); }
extern "C" int64_t host_first_slot(int i, int f) { return qssm_sscan::first_slot(i, f); }
extern "C" int64_t host_most(int64_t tokens, int64_t waves) { return qssm_sscan::most_slots(tokens, waves); }
extern "C" int64_t host_slots(int64_t tokens, int64_t nseq, int64_t piece) { return qssm_sscan::carry_slots(tokens, nseq, piece); }
