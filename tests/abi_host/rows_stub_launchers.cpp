// Stand-in launchers of the rows' operators and of the verification of drafts
// for the host-only build of their argument checks (rows_api.cpp, no HIP
// runtime): each counts the call and keeps its arguments.
#include "../../gguf_block_quantized_qmv_amd/csrc/rows_internal.h"

namespace stub {
int launches = 0;
qmv::SortArgs sort{};
qmv::MoveArgs move{};
qmv::LoraArgs lora{};
qmv::VerifyArgs verify{};
}  // namespace stub

namespace qmv {

int launch_rows_sort(const SortArgs &a, void *) { stub::sort = a; return ++stub::launches, 0; }
int launch_rows_spread(const MoveArgs &a, void *) { stub::move = a; return ++stub::launches, 0; }
int launch_rows_combine(const MoveArgs &a, void *) { stub::move = a; return ++stub::launches, 0; }
int launch_rows_combine_grad(const MoveArgs &a, void *) { stub::move = a; return ++stub::launches, 0; }
int launch_lora(const LoraArgs &a, void *) { stub::lora = a; return ++stub::launches, 0; }
int launch_verify_drafts(const VerifyArgs &a, void *) { stub::verify = a; return ++stub::launches, 0; }

}  // namespace qmv
