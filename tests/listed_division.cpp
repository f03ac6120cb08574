// The walk of attn_division.cpp over plans as a launch over listed blocks makes
// them: parts of fewer records than those of the whole attention.  lens: 16 for
// every listed record.
#include "w4_attn_plan.cuh"

namespace {

w4::Plan listed_plan(int D, int NT, int rows, int record_bytes) {
    const bool bf16 = record_bytes == 64 * D;             // the formats' sizes differ
    return w4::plan_of(D, NT, rows, record_bytes, w4::listed_part(bf16, D));
}

}  // namespace

#define plan_of listed_plan
#include "attn_division.cpp"
