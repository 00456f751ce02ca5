// Stage 1's instances for the own part of a shared-prefix decode, which run
// beside the prefix pass (see BESIDE in stage1.cu); a translation unit of their
// own, compiled in parallel with the others.
#define PD_STAGE1_BESIDE 1
#include "stage1.cu"
