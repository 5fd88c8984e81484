import os,sys; sys.path.insert(0,'/root/repo/_work'); 
import torch
sys.path.insert(0,os.getcwd())
from fully_sharded_unit_gb300 import binding as B
assert 'fork' in B.__file__, B.__file__
from probe_gemm import run
os.environ["PROBE_SHARE"]="0"
import io,contextlib
for lay in ("out_in","in_out"):
  for bn in (256,224,192,160,128,96,64):
    os.environ["PROBE_BN"]=str(bn)
    res=[]
    N=bn*4*5
    for K in (1280,5120):
        with contextlib.redirect_stdout(io.StringIO()):
            us=run(4864,K,N,"fwd",lay)    # 19 x 20 tiles = 5 rounds
        res.append(us)
    slope=(res[1]-res[0])/5/60   # us per stage
    print(lay,bn,"us",["%.1f"%r for r in res],"stage us %.4f  cycles@1.93 %.0f ideal %d"%(slope,slope*1930,2*bn), "per tile at 1280: %.2f"%(res[0]/5), "TF %.0f"%(2*4864*5120*N/res[1]/1e6),flush=True)
