// Host side of the few-rows product (few.hip).
#pragma once

#include "epilogue.hpp"

namespace moonep {

// Whether a product over `nranks` ranks' rows goes to the few-rows kernel.
bool few_rows(const moe_cfg* c, bool dense, int64_t nranks, int cus);

// Bytes of workspace that any such call of this configuration needs.
size_t few_ws_bytes(const moe_cfg* c);

// Launches it (arguments checked); cu null: every row belongs to one matrix.
int launch_few(const moe_cfg* c, const uint16_t* x, const uint16_t* w_home, const uint16_t* w_pref,
               const int32_t* cu, const Epilogue& ep, int rank_begin, int rank_end, void* workspace,
               hipStream_t stream);

// Bytes of workspace of the epilogue's backward (epilogue.hip).
size_t epilogue_bwd_ws_bytes(const moe_cfg* c);

}  // namespace moonep
