// The choice of kernels for a dense linear's calls (dense_api.cpp), from the
// types and sizes alone. Host code, no HIP call.
#pragma once

#include "kernels.h"

namespace poetx {

struct FwdChoice {
  bool stream;          // the streaming kernel, and nothing below
  bool dense;           // the 256 x 256 tiles, else `tile`
  bool widen, w_tiled;  // INT8 codes widened into the workspace (in the tiled layout)
  TilePlan tile;
  // whether a launch takes the tiles of y
  bool launchable() const { return stream || dense || tile.nsplit != 0; }
};
FwdChoice choose_fwd(DType t, bool int8, int64_t tokens, int64_t d_in, int64_t d_out);

struct BwdChoice {
  bool dense;       // g_x on the 256 x 256 tiles, else `gx`
  bool paired;      // g_x and g_W, where both are asked for, in one launch
  TilePlan gx, gw;
  TilePairPlan pair;
  bool gx_launchable() const { return dense || gx.nsplit != 0; }
  bool gw_launchable() const { return gw.nsplit != 0; }
};
BwdChoice choose_bwd(DType t, bool int8, int64_t tokens, int64_t d_in, int64_t d_out);

}  // namespace poetx
